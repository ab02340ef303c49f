"""Plans of int8 products over experts on the CPU: what a call gets does not hang on the calls before it."""
import pytest

import quantized_gemm_bf16_amd as qg

FAKE = 1 << 20
W8A8 = (qg.QUANT_BLOCK_F32, 0, 1, 0)


def plan(g, stride, pitch=7168, m=16384, n=2048, k=7168, e=64):
    kw = dict(num=e, offsets=FAKE)
    return g.plan(qg.operation(quant_a=W8A8, quant_b=W8A8), qg.layout("i8", m, k, ld=pitch, **kw), qg.layout("f32", m, 1, **kw),
                  qg.layout("i8", n, k, ld=pitch, num=e, stride=stride), qg.layout("f32", n, 1, num=e, stride=n if stride else 0), None,
                  qg.layout("bf16", m, n, **kw), 1.0, 0.0)


# weights of each expert (0.9 GB, past the memory-side cache), one matrix for all (132 MB with A's), and that at three times the pitch (past it)
CALLS = [(2048 * 7168, 7168), (0, 7168), (0, 3 * 7168)]


@pytest.mark.parametrize("order", [(0, 1, 2), (2, 1, 0), (1, 2, 0), (1, 0, 2)])
def test_plans_in_any_order(order):
    alone = [plan(qg.Gemm(), *c) for c in CALLS]
    assert alone[0] != alone[1] and alone[0] == alone[2]  # the rule looks at the operands' size
    g = qg.Gemm()
    for i in order + order:
        assert plan(g, *CALLS[i]) == alone[i], (order, i)
