"""Raw device addresses in the binding's calls: an int of any kind, a subclass's too. On the CPU, and no call here reaches a launch
(an address that is not aligned is refused)."""
import enum

import pytest

import quantized_gemm_bf16_amd as qg


class Buffer(enum.IntEnum):
    A = 1 << 20
    ODD = (1 << 20) + 2


class Address(int):
    pass


KINDS = [int, Address, Buffer]
W8A8 = (qg.QUANT_BLOCK_F32, 0, 1, 0)


@pytest.mark.parametrize("kind", KINDS)
def test_addresses(kind):
    """Well-formed calls with one address that is not aligned: that is what they are refused for."""
    g, p, odd = qg.Gemm(), kind(1 << 20), kind((1 << 20) + 2)
    x, q, s = qg.layout("bf16", 4, 64), qg.layout("i8", 4, 64), qg.layout("f32", 4, 1)
    al = qg.ERR_ALIGNMENT
    op = qg.operation(epilogue=qg.EPI_BIAS, bias=p)
    d = qg.layout("bf16", 4, 4, ld=8)
    assert op.epi.bias == 1 << 20
    assert g.run_raw(op, 1.0, p, x, None, None, p, x, None, None, 0.0, None, None, odd, d, None) == al
    w8 = qg.operation(quant_a=W8A8, quant_b=W8A8)
    assert g.run_raw(w8, 1.0, p, q, odd, s, p, q, p, s, 0.0, None, None, p, d, None) == al
    mq, ms = qg.layout("e2m1", 4, 64), qg.layout("e8m0", 4, 2)
    assert g.mx_quantize_raw(p, x, odd, mq, p, ms, rows=p) == al and g.mx_dequantize_raw(p, mq, p, ms, odd, x) == al
    assert g.int_quantize_raw(p, x, odd, q, p, s, rows=p) == al and g.int_dequantize_raw(p, q, odd, s, p, x) == al
    ids, w = qg.layout("i32", 4, 2), qg.layout("f32", 4, 2)
    assert g.route_raw(qg.routing(top_k=2), p, x, p, odd, ids, p, w) == al and g.route_raw(qg.routing(top_k=2), p, x, odd, p, ids, p, w) == al
    assert g.group_rows_raw(8, p, ids, p, p, odd) == al and g.group_rows_raw(8, odd, ids, p, p, p) == al
    r = qg.layout("bf16", 8, 64)
    assert g.combine_raw(p, r, odd, p, w, p, x) == al and g.combine_raw(p, r, p, odd, w, p, x, beta=1.0, C=p, Cd=x) == al
